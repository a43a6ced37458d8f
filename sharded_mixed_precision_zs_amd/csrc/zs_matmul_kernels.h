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
 *
 * Sums. The unit adds eight neighbouring products before it adds them to an
 * fp32 sum, and keeps of them what lies within some 13 bits of the largest.
 * E2M1 products span less. E4M3 elements reach from 448 down to 2^-9, so an A
 * in E4M3 is multiplied in two halves, elements from 2 on and elements below
 * 2, zeros in the others' places: products of the first are multiples of 2^-3
 * below 2^12, of the second multiples of 2^-10 below 2^4, and nothing of
 * either is dropped (every code of a half against every code of B, and
 * results left by cancellation, come out exactly). One half at once differed
 * by up to 3e-4 of the sum of magnitudes. It costs twice the matrix
 * instructions, which is what 16-bit operands would cost.
 */
#ifndef ZS_MATMUL_KERNELS_H
#define ZS_MATMUL_KERNELS_H

#include "zs_epilogue.h"

namespace zs {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct MatmulArgs {
  const uint8_t *a, *as, *b, *bs;
  void *c;
  uint64_t ldc;
  uint32_t m, n, padded;   /* padded: K rounded up to whole groups */
  float *part;             /* tiles split along K: [splits][m][n] sums */
  uint32_t split_groups;   /* groups of a split, a multiple of four; all: one split */
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

/* ------------------------------------------------------------------------
 * Tiles of C through LDS. A block of NW waves, in two rows, computes BM x BN,
 * in stages of 256 elements of K that two LDS buffers hold in turn: while the
 * matrix cores work on one, the loads of the next stage go straight to the
 * other, so a stage's arithmetic hides its loads.
 *
 * The large tiles, 256 x 256 of 4 x 4 bits in eight waves and 128 x 256 of
 * 8 x 4 in four, are as large as two buffers in LDS and the sums in registers
 * allow, for a fragment read from LDS serves FM or FN matrix instructions:
 * 8192^3 of 4 x 4 bits 275 us (4.0 PFLOP/s), 8192 x 4096 x 4096 of 4 x 4
 * bits 78 us (in four waves 83), of 8 x 4 bits 222 us (1.24 PFLOP/s; twice
 * that of the instructions, for A's two halves). At 8192^3 of 4 x 4 bits the
 * matrix cores work half of the cycles, at 1.75 GHz under that load; a fifth
 * of the waves' time goes into the barrier of a stage. 128 x 128 in four waves
 * for what gives fewer tiles than CUs: 77 x 50257 x 768 of 4 x 4 bits, fp16:
 * 8.6 us.
 *
 * LDS rows are 128 bytes: 256 E2M1 elements, or 128 E4M3 elements (A then
 * has two planes). A wave's load fills 8 such rows, 16 bytes a lane, whole
 * lines of memory; the 16-byte piece c of row r lies at c ^ x(r), x(r) =
 * r % 8 with its lowest bit flipped in every other 8 rows, so that the lanes
 * of a fragment, which read the same piece of 32 rows, meet no bank twice in
 * any 8 or 16 of them.
 *
 * Scales: a thread fetches 16 bytes of a row or two, those of 512 elements,
 * and puts them into LDS a chunk ahead; a fragment's lane then reads the 8
 * bytes of a stage.
 * ---------------------------------------------------------------------- */
constexpr uint32_t kStageK = 256;                 /* elements of K per stage */
constexpr uint32_t kStageGroups = kStageK / kMxGroup;

typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void global_void;

__device__ __forceinline__ uint32_t swizzle(uint32_t row) { return (row ^ (row >> 3 & 1)) & 7; }

/* 16 bytes per lane from memory to LDS: lane l's go to dst + 16 l. */
__device__ __forceinline__ void load_lds16(const uint8_t *src, uint8_t *dst) {
  __builtin_amdgcn_global_load_lds((global_void *)src, (lds_void *)dst, 16, 0, 0);
}

/* A barrier behind which every wave's loads to LDS are there. The barrier
 * itself does not promise that: it orders what a wave has waited for. */
__device__ __forceinline__ void loads_barrier() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
}

template <int AF>
__device__ __forceinline__ f32x16 mfma(const i32x8 &b, const i32x8 &a, f32x16 acc, uint32_t sb,
                                       uint32_t sa, bool high) {
  /* the lane's scale is byte 0 (first 64 elements of a group) or 2 of a word */
  return high ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, acc, 4, kMfmaFormat<AF>, 2,
                                                                sb, 2, sa)
              : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, acc, 4, kMfmaFormat<AF>, 0,
                                                                sb, 0, sa);
}

/* The elements of magnitude 2 and above, whose highest exponent bit is set
 * (NaN codes are among them), zeros for the others; the other way round with
 * other = ~0. The byte permute's selectors 8 to 11 spread a sign bit: those
 * of bytes 1 and 3 of either word. */
__device__ __forceinline__ i32x8 upper_half(const i32x8 &a, uint32_t other = 0) {
  i32x8 h;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t w = (uint32_t)a[j];
    h[j] = (int)(w & (__builtin_amdgcn_perm(w << 1, w << 9, 0x0b090a08u) ^ other));
  }
  return h;
}

__device__ __forceinline__ void put4(i32x8 &f, int at, const u32x4 &w) {
#pragma unroll
  for (int j = 0; j < 4; ++j) f[at + j] = (int)w[j];
}

/* One step's operands: 64 elements of K of a wave's rows, as read. */
template <int AF>
constexpr int kHalves = AF == ZS_MX_E2M1 ? 1 : 2;   /* 16-byte pieces of A */

template <int AF, int FM, int FN>
struct Fragments {
  u32x4 a[FM][kHalves<AF>], b[FN];
};

/* 16-byte piece c of LDS row `row` (128 bytes); x = swizzle(row). */
__device__ __forceinline__ u32x4 piece(const uint8_t *lds, uint32_t row, uint32_t c, uint32_t x) {
  return *reinterpret_cast<const u32x4 *>(lds + row * 128 + ((c ^ x) * 16));
}

template <int AF, int FM, int FN>
__device__ __forceinline__ void read_step(const uint8_t *sa, const uint8_t *sb, int ks,
                                          uint32_t plane, uint32_t row, uint32_t g, uint32_t x,
                                          Fragments<AF, FM, FN> &f) {
#pragma unroll
  for (int j = 0; j < FN; ++j) f.b[j] = piece(sb, j * 32 + row, 2 * ks + g, x);
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    if constexpr (AF == ZS_MX_E2M1) {
      f.a[i][0] = piece(sa, i * 32 + row, 2 * ks + g, x);
    } else {
      const uint8_t *q = sa + (ks >> 1) * plane;
      f.a[i][0] = piece(q, i * 32 + row, 4 * (ks & 1) + g, x);
      f.a[i][1] = piece(q, i * 32 + row, 4 * (ks & 1) + 2 + g, x);
    }
  }
}

/* A stage's scales of a wave's rows, a word per group. */
template <int FM, int FN>
struct StageScales {
  uint32_t a[FM][2], b[FN][2];
};

template <int FM, int FN>
__device__ __forceinline__ void read_scales(const uint8_t *sa, const uint8_t *sb, uint32_t row,
                                            uint32_t g, StageScales<FM, FN> &w) {
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const u32x2 v = *reinterpret_cast<const u32x2 *>(sa + (i * 32 + row) * 16);
    w.a[i][0] = v.x >> (8 * g);
    w.a[i][1] = v.y >> (8 * g);
  }
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const u32x2 v = *reinterpret_cast<const u32x2 *>(sb + (j * 32 + row) * 16);
    w.b[j][0] = v.x >> (8 * g);
    w.b[j][1] = v.y >> (8 * g);
  }
}

template <int AF, int FM, int FN>
__device__ __forceinline__ void multiply_step(const Fragments<AF, FM, FN> &f, int ks,
                                              const StageScales<FM, FN> &w,
                                              f32x16 (&acc)[FM][FN]) {
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    i32x8 a{};
    put4(a, 0, f.a[i][0]);
    if constexpr (AF == ZS_MX_E4M3) put4(a, 4, f.a[i][1]);
    const i32x8 first = AF == ZS_MX_E4M3 ? upper_half(a) : a;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      i32x8 b{};
      put4(b, 0, f.b[j]);
      acc[i][j] = mfma<AF>(b, first, acc[i][j], w.b[j][ks >> 1], w.a[i][ks >> 1], ks & 1);
    }
    if constexpr (AF == ZS_MX_E4M3) {
      const i32x8 second = a ^ first;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        i32x8 b{};
        put4(b, 0, f.b[j]);
        acc[i][j] = mfma<AF>(b, second, acc[i][j], w.b[j][ks >> 1], w.a[i][ks >> 1], ks & 1);
      }
    }
  }
}

/* Asks the scheduler to spread a step's LDS reads among the matrix
 * instructions of the step before. */
template <int AF, int FM, int FN>
__device__ __forceinline__ void interleave() {
  constexpr int reads = FN + FM * kHalves<AF>, products = FM * FN * kHalves<AF>;
  constexpr int each = products / reads > 0 ? products / reads : 1;
#pragma unroll
  for (int i = 0; i < reads; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, each, 0);   /* matrix instructions */
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);      /* an LDS read */
  }
  __builtin_amdgcn_sched_barrier(0);   /* nothing moves into another step */
}

/* Result element types by their size and rounding. */
template <int CDT>
__device__ __forceinline__ void put_c4(uint8_t *lds, const float (&x)[4]) {
  if constexpr (CDT == ZS_FP32)
    *reinterpret_cast<float4 *>(lds) = make_float4(x[0], x[1], x[2], x[3]);
  else
    *reinterpret_cast<u32x2 *>(lds) = u32x2{pack2<CDT>(x[0], x[1]), pack2<CDT>(x[2], x[3])};
}

template <int V>
struct Const {
  static constexpr int value = V;
};

template <int AF, int CDT, int BM, int BN, int NW, class E>
__global__ __launch_bounds__(64 * NW, NW / 4) void matmul_tile_kernel(MatmulArgs p, E epilogue) {
  constexpr int kAcross = NW / 2, kThreads = 64 * NW;   /* two rows of NW / 2 waves */
  constexpr int FM = BM / 64, FN = BN / (32 * kAcross); /* 32 x 32 fragments per wave */
  constexpr int LA = BM / (8 * NW), LB = BN / (8 * NW); /* loads of 8 rows per wave */
  constexpr uint32_t kPlanes = AF == ZS_MX_E2M1 ? 1 : 2, kPlane = BM * 128;
  __shared__ __align__(16) uint8_t sa0[kPlanes * kPlane], sa1[kPlanes * kPlane];
  __shared__ __align__(16) uint8_t sb0[BN * 128], sb1[BN * 128];
  __shared__ __align__(16) uint8_t scales[2 * (BM + BN) * 16];   /* two chunks' */
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const uint32_t r = lane & 31, g = lane >> 5;
  /* its corner of the tile */
  const uint32_t tm = wave / kAcross * (BM / 2), tn = wave % kAcross * (BN / kAcross);

  /* Blocks go round the eight XCDs; each XCD takes a run of tiles, and runs
   * walk groups of eight tile rows, so that its L2 sees the same operands
   * again soon. */
  const uint32_t tiles_m = (p.m + BM - 1) / BM, tiles_n = (p.n + BN - 1) / BN;
  const uint32_t total = tiles_m * tiles_n;
  uint32_t id = blockIdx.x;
  {
    const uint32_t per = total / 8, extra = total % 8, xcd = id % 8, at = id / 8;
    id = xcd * per + (xcd < extra ? xcd : extra) + at;
  }
  constexpr uint32_t kBand = 8;
  const uint32_t band = id / (kBand * tiles_n), in_band = id % (kBand * tiles_n);
  const uint32_t high = tiles_m - band * kBand < kBand ? tiles_m - band * kBand : kBand;
  const uint32_t m0 = (band * kBand + in_band % high) * BM, n0 = (in_band / high) * BN;

  const uint64_t row_a = mx_bytes<AF>(p.padded), row_b = p.padded / 2;
  const uint32_t scale_row = p.padded / kMxBlock;
  const uint32_t group0 = blockIdx.y * p.split_groups;   /* this split's share of K */
  const uint32_t left = p.padded / kMxGroup - group0;
  const uint32_t groups = left < p.split_groups ? left : p.split_groups;
  const uint8_t *ta = p.a + m0 * row_a + mx_bytes<AF>((uint64_t)group0 * kMxGroup);
  const uint8_t *tb = p.b + n0 * row_b + (uint64_t)group0 * (kMxGroup / 2);

  /* Rows past the last are read as the last; their results are not stored. */
  const uint32_t last_a = p.m - 1 - m0, last_b = p.n - 1 - n0;
  uint32_t off_a[LA], off_b[LB];
#pragma unroll
  for (int i = 0; i < LA; ++i) {
    const uint32_t row = (wave * (LA) + i) * 8 + lane / 8;
    off_a[i] = (row < last_a ? row : last_a) * (uint32_t)row_a + ((lane & 7) ^ swizzle(row)) * 16;
  }
#pragma unroll
  for (int i = 0; i < LB; ++i) {
    const uint32_t row = (wave * (LB) + i) * 8 + lane / 8;
    off_b[i] = (row < last_b ? row : last_b) * (uint32_t)row_b + ((lane & 7) ^ swizzle(row)) * 16;
  }
  /* this thread's rows of scales: A's, then B's */
  constexpr int kScaleRows = (BM + BN + kThreads - 1) / kThreads;
  const uint8_t *scale_of[kScaleRows];
#pragma unroll
  for (int i = 0; i < kScaleRows; ++i) {
    const uint32_t t = threadIdx.x + i * kThreads, rb = t - BM;
    scale_of[i] = (t < BM ? p.as + (uint64_t)(m0 + (t < last_a ? t : last_a)) * scale_row
                          : p.bs + (uint64_t)(n0 + (rb < last_b ? rb : last_b)) * scale_row) +
                  group0 * 4;
  }

  /* Bit i: the lane's piece of its i-th row lies in the upper half of a line. */
  uint32_t upper_a = 0, upper_b = 0;
#pragma unroll
  for (int i = 0; i < LA; ++i)
    upper_a |= ((((lane & 7) ^ swizzle((wave * (LA) + i) * 8 + lane / 8)) >> 2) & 1) << i;
#pragma unroll
  for (int i = 0; i < LB; ++i)
    upper_b |= ((((lane & 7) ^ swizzle((wave * (LB) + i) * 8 + lane / 8)) >> 2) & 1) << i;

  /* A stage of one group only (the last, where the groups are odd) loads the
   * half of each row that it has twice, rather than past the row's end. A
   * stage past the last loads the last again: no branch parts the loop. */
  const uint32_t stages = (groups + kStageGroups - 1) / kStageGroups;
  auto load = [&](uint32_t stage, uint8_t *sa, uint8_t *sb) {
    stage = stage < stages ? stage : stages - 1;
    const bool half = (stage + 1) * kStageGroups > groups;
    const uint8_t *qa = ta + mx_bytes<AF>((uint64_t)stage * kStageK);
    const uint8_t *qb = tb + (uint64_t)stage * (kStageK / 2);
    const uint32_t mask = half ? ~0u : 0u;
    const uint32_t ua = kPlanes == 1 ? upper_a & mask : 0, ub = upper_b & mask;
#pragma unroll
    for (uint32_t pl = 0; pl < kPlanes; ++pl)
#pragma unroll
      for (int i = 0; i < LA; ++i)
        load_lds16((half ? qa : qa + pl * 128) + (off_a[i] - ((ua >> i) & 1) * 64),
                   sa + pl * kPlane + (wave * (LA) + i) * 1024);
#pragma unroll
    for (int i = 0; i < LB; ++i)
      load_lds16(qb + (off_b[i] - ((ub >> i) & 1) * 64), sb + (wave * (LB) + i) * 1024);
  };

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{};
  /* Scales go a chunk of four groups at a time, from no further than the
   * row's last four; a last chunk that starts later is shifted down. */
  struct __attribute__((packed, aligned(4))) W4 { uint32_t w[4]; };
  uint32_t raw[kScaleRows][4];
  auto fetch_scales = [&](uint32_t group) {
    const uint32_t at = group + 4 <= groups ? group : groups >= 4 ? groups - 4 : 0;
#pragma unroll
    for (int i = 0; i < kScaleRows; ++i) {
      if ((BM + BN) % kThreads && threadIdx.x + i * kThreads >= BM + BN) break;
      const W4 v = *reinterpret_cast<const W4 *>(scale_of[i] + at * 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) raw[i][k] = v.w[k];
    }
  };
  auto put_scales = [&](uint32_t group, uint32_t chunk) {
    const uint32_t late = group + 4 > groups && groups >= 4 ? group + 4 - groups : 0;   /* <= 3 */
#pragma unroll
    for (int i = 0; i < kScaleRows; ++i) {
      if ((BM + BN) % kThreads && threadIdx.x + i * kThreads >= BM + BN) break;
      u32x4 v = {raw[i][0], raw[i][1], raw[i][2], raw[i][3]};
      v = late & 1 ? u32x4{v.y, v.z, v.w, v.w} : v;
      v = late & 2 ? u32x4{v.z, v.w, v.w, v.w} : v;
      *reinterpret_cast<u32x4 *>(scales + chunk + (threadIdx.x + i * kThreads) * 16) = v;
    }
  };

  /* Fragments start at multiples of 16 rows, which leave x(r) as it is. The
   * operands of step k + 1 are read while step k multiplies. A stage's last
   * step stands behind the barrier: by then every wave holds what it needs
   * of this buffer, and the other one, asked for a stage ago, is complete;
   * so the next stage's first operands and the loads after it are on their
   * way before this stage's last products. */
  const uint32_t x = swizzle(r);
  const uint32_t full = groups / kStageGroups;    /* stages of two groups */
  Fragments<AF, FM, FN> f0, f1;
  StageScales<FM, FN> w0, w1;
  constexpr uint32_t kChunk = (BM + BN) * 16;
  const uint32_t srow_a = tm * 16, srow_b = (BM + tn) * 16;   /* the wave's rows of scales */
  auto run_stage = [&](uint8_t *sa, uint8_t *sb, const uint8_t *next_sa, const uint8_t *next_sb,
                       uint32_t next_sc, uint32_t stage, const StageScales<FM, FN> &w,
                       StageScales<FM, FN> &next_w, auto first, uint32_t put_sc) {
    const uint8_t *qa = sa + tm * 128, *qb = sb + tn * 128;
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (decltype(first)::value) fetch_scales((stage + 2) * kStageGroups);
    read_step<AF, FM, FN>(qa, qb, 1, kPlane, r, g, x, f1);
    multiply_step<AF, FM, FN>(f0, 0, w, acc);
    interleave<AF, FM, FN>();
    read_step<AF, FM, FN>(qa, qb, 2, kPlane, r, g, x, f0);
    multiply_step<AF, FM, FN>(f1, 1, w, acc);
    interleave<AF, FM, FN>();
    read_step<AF, FM, FN>(qa, qb, 3, kPlane, r, g, x, f1);
    multiply_step<AF, FM, FN>(f0, 2, w, acc);
    interleave<AF, FM, FN>();
    loads_barrier();
    __builtin_amdgcn_sched_barrier(0);
    /* past the last stage, what is loaded and read here is not used */
    read_step<AF, FM, FN>(next_sa + tm * 128, next_sb + tn * 128, 0, kPlane, r, g, x, f0);
    read_scales<FM, FN>(scales + next_sc + srow_a, scales + next_sc + srow_b, r, g, next_w);
    load(stage + 2, sa, sb);
    if constexpr (decltype(first)::value) put_scales((stage + 2) * kStageGroups, put_sc);
    multiply_step<AF, FM, FN>(f1, 3, w, acc);
    __builtin_amdgcn_sched_barrier(0);
  };

  if (stages) {
    load(0, sa0, sb0);
    if (groups >= 4) {
      fetch_scales(0);
    } else {   /* shorter rows, of a single chunk, a word at a time */
#pragma unroll
      for (int i = 0; i < kScaleRows; ++i) {
        if ((BM + BN) % kThreads && threadIdx.x + i * kThreads >= BM + BN) break;
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k)
          raw[i][k] = *reinterpret_cast<const uint32_t *>(scale_of[i] +
                                                          4 * (k < groups ? k : groups - 1));
        scale_of[i] = p.a;   /* what the loop fetches is not used: 16 bytes that are there */
      }
    }
    put_scales(0, 0);
    loads_barrier();
    load(1, sa1, sb1);
    read_scales<FM, FN>(scales + srow_a, scales + srow_b, r, g, w0);
    read_step<AF, FM, FN>(sa0 + tm * 128, sb0 + tn * 128, 0, kPlane, r, g, x, f0);
  }
  uint32_t sc = 0, s = 0;   /* a chunk's scales: two stages' */
  for (; s + 1 < full; s += 2, sc ^= kChunk) {
    run_stage(sa0, sb0, sa1, sb1, sc + 8, s, w0, w1, Const<true>{}, sc ^ kChunk);
    run_stage(sa1, sb1, sa0, sb0, sc ^ kChunk, s + 1, w1, w0, Const<false>{}, 0);
  }
  if (s < full) run_stage(sa0, sb0, sa1, sb1, sc + 8, s, w0, w1, Const<true>{}, sc ^ kChunk);
  if (groups % kStageGroups) {   /* half a stage left: its first operands are in f0 */
    const bool odd = full & 1;
    read_step<AF, FM, FN>((odd ? sa1 : sa0) + tm * 128, (odd ? sb1 : sb0) + tn * 128, 1, kPlane, r,
                          g, x, f1);
    if (odd) w0 = w1;
    multiply_step<AF, FM, FN>(f0, 0, w0, acc);
    multiply_step<AF, FM, FN>(f1, 1, w0, acc);
  }
  loads_barrier();   /* the strips below take the place of what was loaded last */

  /* Each wave turns strips of 32 rows round in its own part of LDS, so that
   * rows of C go out in runs: 16-byte pieces, swizzled as above. With an
   * epilogue the strips are fp32, and a lane finishes eight results. */
  constexpr int SDT = E::kOn ? ZS_FP32 : CDT;   /* the strips' type */
  constexpr uint32_t kEsz = SDT == ZS_FP32 ? 4 : 2, kRow = FN * 32 * kEsz, kPieces = kRow / 16;
  static_assert(32 * kRow * kAcross <= sizeof(sa0) && 32 * kRow * kAcross <= sizeof(sb0),
                "strips fit");
  uint8_t *strip = (wave / kAcross ? sb0 : sa0) + wave % kAcross * 32 * kRow;
  uint8_t *c = static_cast<uint8_t *>(p.c);
  uint64_t ldc = p.ldc;
  if (p.part) {   /* CDT is fp32 then */
    c = reinterpret_cast<uint8_t *>(p.part + (uint64_t)blockIdx.y * p.m * p.n);
    ldc = p.n;
  }
  const bool vec = ((uintptr_t)c & 15) == 0 && ldc * kEsz % 16 == 0;
  /* An epilogue's lane: eight columns of every kRows-th row; its residual's
   * vectors of a strip are on their way while the strip is turned. */
  constexpr uint32_t kAhead = FN * 4, kRows = 64 / kAhead, kStrips = 32 / kRows;
  const uint32_t pc = lane % kAhead, col = n0 + tn + pc * 8;
  float bias[8] = {};
  if constexpr (E::kOn) {
    if (epilogue.bias) load8<CDT, false>(epilogue.bias, col, p.n, bias);
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    Raw16<8> residual[kStrips];
    if constexpr (E::kOn) {
      if (epilogue.res) {
#pragma unroll
        for (uint32_t k = 0; k < kStrips; ++k) {
          const uint32_t row = m0 + tm + i * 32 + k * kRows + lane / kAhead;
          residual[k] = epilogue.load(row < p.m ? row : p.m - 1, col, p.n);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                            acc[i][j][4 * q + 3]};
        const uint32_t byte = (j * 32 + q * 8 + g * 4) * kEsz;
        put_c4<SDT>(strip + r * kRow + (((byte / 16) ^ (r % kPieces)) * 16) + byte % 16, v);
      }
    __builtin_amdgcn_wave_barrier();
    const uint32_t col0 = n0 + tn;
    if constexpr (E::kOn) {
#pragma unroll
      for (uint32_t k = 0; k < kStrips; ++k) {
        const uint32_t lr = k * kRows + lane / kAhead, row = m0 + tm + i * 32 + lr;
        float v[8];
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
          const float4 w = *reinterpret_cast<const float4 *>(
              strip + lr * kRow + (((2 * pc + h) ^ (lr % kPieces)) * 16));
          v[4 * h] = w.x;
          v[4 * h + 1] = w.y;
          v[4 * h + 2] = w.z;
          v[4 * h + 3] = w.w;
        }
        if (row < p.m)
          epilogue.template store<CDT>(row, col, p.n, v, bias, residual[k],
                                       static_cast<uint16_t *>(p.c), p.ldc);
      }
      __builtin_amdgcn_wave_barrier();
      continue;
    }
    constexpr uint32_t kRowsAtOnce = 64 / kPieces > 0 ? 64 / kPieces : 1;
#pragma unroll
    for (uint32_t k = 0; k < 32 / kRowsAtOnce; ++k) {
      const uint32_t lr = k * kRowsAtOnce + lane / kPieces, pc = lane % kPieces;
      const uint32_t row = m0 + tm + i * 32 + lr, col = col0 + pc * (16 / kEsz);
      const uint8_t *from = strip + lr * kRow + ((pc ^ (lr % kPieces)) * 16);
      const u32x4 w = *reinterpret_cast<const u32x4 *>(from);
      if (row >= p.m) continue;
      uint8_t *out = c + ((uint64_t)row * ldc + col) * kEsz;
      if (col + 16 / kEsz <= p.n) {
        if (vec) *reinterpret_cast<u32x4 *>(out) = w;
        else *reinterpret_cast<Loose16 *>(out) = Loose16{{w.x, w.y, w.z, w.w}};
      } else {
        for (uint32_t e = 0; col + e < p.n; ++e) {
          if constexpr (kEsz == 4)
            reinterpret_cast<uint32_t *>(out)[e] = reinterpret_cast<const uint32_t *>(from)[e];
          else
            reinterpret_cast<uint16_t *>(out)[e] = reinterpret_cast<const uint16_t *>(from)[e];
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

/* The splits' sums, added in order and rounded once: a thread per result, its
 * sums still in the caches (768 x 768 x 8192 of 8 x 4 bits in six pieces: 24
 * us both launches, one piece 53). */
template <int CDT, class E>
__global__ __launch_bounds__(kBlock) void matmul_join_kernel(MatmulArgs p, uint32_t splits,
                                                             E epilogue) {
  const uint64_t id = (uint64_t)blockIdx.x * kBlock + threadIdx.x, all = (uint64_t)p.m * p.n;
  if (id >= all) return;
  float s = 0.0f;
  for (uint32_t k = 0; k < splits; ++k) s += p.part[k * all + id];
  const uint32_t row = (uint32_t)(id / p.n), col = (uint32_t)(id % p.n);
  if constexpr (E::kOn)
    epilogue.template store1<CDT>(row, col, p.n, s, static_cast<uint16_t *>(p.c), p.ldc);
  else if constexpr (CDT == ZS_FP32) static_cast<float *>(p.c)[row * p.ldc + col] = s;
  else static_cast<uint16_t *>(p.c)[row * p.ldc + col] = pack1<CDT>(s);
}

/* ------------------------------------------------------------------------
 * Few rows of A (m <= 32): bound by reading B once. A block owns 32 rows
 * of B; its eight waves share K in pieces of 256 elements and join in wave
 * order. B goes through LDS, a wave's piece in its own part, so that a load
 * takes whole lines (eight lanes to a row's 128 bytes; straight to registers
 * an instruction would touch 32 rows for 32 bytes each): two parts in turn,
 * and no barrier but a wave's own wait for its loads. A comes from the caches.
 * PAIR, for the fewest rows of an 8-bit A: its two halves are rows r and
 * r + 16 of one instruction, and are added with the waves' sums.
 * One row by 32000 x 4096, 8 x 4 bits: 14.4 us, 4.9 TB/s of the 70 MB of B,
 * 2 us of it the launch; taking A's halves apart is 1.5 us of it. (B straight
 * to registers cost 4 us more.)
 * ---------------------------------------------------------------------- */
constexpr int kThinWaves = 8;
constexpr uint32_t kThinPart = 32 * 128;   /* a piece: 32 rows of 128 bytes */

template <int AF, int CDT, bool PAIR, class E>
__global__ __launch_bounds__(64 * kThinWaves, 4) void matmul_thin_kernel(MatmulArgs p, int vec,
                                                                         E epilogue) {
  /* staging, then the waves' sums in its place */
  constexpr uint32_t kSums = kThinWaves * 16 * 64 * 4, kStage = kThinWaves * kThinPart;
  __shared__ __align__(16) uint8_t stage0[kStage], stage1[kStage];
  static_assert(kSums <= kStage, "the sums fit");
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const uint32_t r = lane & 31, g = lane >> 5, n0 = blockIdx.x * 32;
  const uint32_t last = p.n - 1 - n0;   /* rows past it are read as it */
  const uint64_t row_b = p.padded / 2;
  const uint32_t scale_row = p.padded / kMxBlock, groups = p.padded / kMxGroup;
  const uint8_t *tb = p.b + n0 * row_b;
  uint32_t off[4], upper = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t row = i * 8 + lane / 8, c = (lane & 7) ^ swizzle(row);
    off[i] = (row < last ? row : last) * (uint32_t)row_b + c * 16;
    upper |= (c >> 2) << i;
  }
  /* a lane's offsets from a wave's bases: below 2^28, for rows take up to 2^22 bytes */
  const uint8_t *bs = p.bs + (uint64_t)n0 * scale_row;
  const uint32_t off_bs = (r < last ? r : last) * scale_row;
  const uint32_t ar = PAIR ? r & 15 : r;
  const uint32_t lower = PAIR && r >= 16 ? ~0u : 0;   /* this lane's half */
  const uint32_t ra = ar < p.m ? ar : p.m - 1;
  const uint32_t off_a = ra * (uint32_t)mx_bytes<AF>(p.padded) + g * 16, off_as = ra * scale_row;
  f32x16 acc{};
  const uint32_t x = swizzle(r), stages = (groups + 1) / 2;
  /* A piece's A and scales go to registers, its B to LDS. A last piece of one
   * group loads what it has twice, and multiplies it once. */
  struct Piece {
    u32x4 a[2][2][kHalves<AF>];
    uint32_t wa[2], wb[2];
  };
  auto load = [&](uint32_t stage, Piece &q, uint8_t *lds) {
#pragma unroll
    for (uint32_t h = 0; h < 2; ++h) {
      const uint32_t group = stage * 2 + h < groups ? stage * 2 + h : groups - 1;
      const uint8_t *a = p.a + mx_bytes<AF>((uint64_t)group * kMxGroup);
      q.wb[h] = *reinterpret_cast<const uint32_t *>(bs + group * 4 + off_bs);
      q.wa[h] = *reinterpret_cast<const uint32_t *>(p.as + group * 4 + off_as);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int v = 0; v < kHalves<AF>; ++v)
          q.a[h][ks][v] = *reinterpret_cast<const u32x4 *>(a + off_a + (ks * kHalves<AF> + v) * 32);
    }
    const uint32_t u = (stage + 1) * 2 > groups ? upper : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      load_lds16(tb + (uint64_t)stage * 128 + (off[i] - ((u >> i) & 1) * 64),
                 lds + wave * kThinPart + i * 1024);
  };
  auto multiply = [&](uint32_t stage, const Piece &q, const uint8_t *lds) {
#pragma unroll
    for (uint32_t h = 0; h < 2; ++h) {
      if (stage * 2 + h >= groups) break;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        i32x8 vb{}, va{};
        put4(vb, 0, piece(lds + wave * kThinPart, r, 4 * h + 2 * ks + g, x));
        put4(va, 0, q.a[h][ks][0]);
        if constexpr (AF == ZS_MX_E4M3) {
          put4(va, 4, q.a[h][ks][1]);
          if constexpr (!PAIR) {
            acc = mfma<AF>(vb, upper_half(va, ~0u), acc, q.wb[h] >> (8 * g), q.wa[h] >> (8 * g),
                           ks & 1);
            __builtin_amdgcn_sched_barrier(0);
          }
          va = upper_half(va, lower);
        }
        acc = mfma<AF>(vb, va, acc, q.wb[h] >> (8 * g), q.wa[h] >> (8 * g), ks & 1);
        if constexpr (AF == ZS_MX_E4M3) __builtin_amdgcn_sched_barrier(0);   /* few registers */
      }
    }
  };
  Piece q0, q1;
  /* Both parts are asked for at once; each is filled again when it is read.
   * The waits are written out: loads to LDS are counted with all others, in
   * order; the last four asked for, the other part's, may be under way still
   * (what the registers wait for, the compiler knows). */
  if (wave < stages) load(wave, q0, stage0);
  if (wave + kThinWaves < stages) load(wave + kThinWaves, q1, stage1);
  for (uint32_t s = wave; s < stages; s += 2 * kThinWaves) {
    if (s + kThinWaves < stages) asm volatile("s_waitcnt vmcnt(4)" ::: "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    multiply(s, q0, stage0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   /* read before it is filled again */
    if (s + 2 * kThinWaves < stages) load(s + 2 * kThinWaves, q0, stage0);
    if (s + kThinWaves < stages) {
      if (s + 2 * kThinWaves < stages) asm volatile("s_waitcnt vmcnt(4)" ::: "memory");
      else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      multiply(s + kThinWaves, q1, stage1);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (s + 3 * kThinWaves < stages) load(s + 3 * kThinWaves, q1, stage1);
    }
  }
  __syncthreads();
  float *sums = reinterpret_cast<float *>(stage0);   /* [wave][16][64] */
#pragma unroll
  for (int e = 0; e < 16; ++e) sums[(wave * 16 + e) * 64 + lane] = acc[e];
  __syncthreads();
  /* a thread takes four neighbouring results: quarter q of lane l */
  const uint32_t q = threadIdx.x / 64, l = threadIdx.x & 63;
  if (q >= 4 || (l & 31) >= p.m) return;
  float v[4] = {0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < kThinWaves; ++w)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] += sums[(w * 16 + q * 4 + e) * 64 + l];
      if constexpr (PAIR) v[e] += sums[(w * 16 + q * 4 + e) * 64 + l + 16];   /* l & 31 < 16 */
    }
  const uint32_t col = n0 + q * 8 + (l >> 5) * 4;
  if constexpr (E::kOn) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      epilogue.template store1<CDT>(l & 31, col + e, p.n, v[e], static_cast<uint16_t *>(p.c),
                                    p.ldc);
  } else {
    store_c4<CDT>(p.c, (uint64_t)(l & 31) * p.ldc, col, p.n, v, vec);
  }
}

}  // namespace zs
#endif  // ZS_MATMUL_KERNELS_H
