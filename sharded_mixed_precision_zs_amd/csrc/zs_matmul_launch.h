/*
 * zs_matmul_launch.h -- the microscaled product's choice of kernel, and its
 * launch. Host code only.
 */
#ifndef ZS_MATMUL_LAUNCH_H
#define ZS_MATMUL_LAUNCH_H

#include "zs_matmul_kernels.h"
#include "zs_ops_common.h"

namespace zs_ops {

using namespace zs;

/* ------------------------------------------------------------------------
 * The product's variant: for few rows of A, bound by B, the thin kernel;
 * the large tiles where they occupy every CU (4096^3 of 4 x 4 bits 42 us,
 * 53 in tiles of 128 x 128; 8 x 4 bits 106 and 120), else 128 x 128 (2048 x
 * 4096 x 4096 of 4 x 4 bits, whose large tiles fill half of the CUs: 29 us,
 * large 36), and where even these leave three CUs of four idle and K is long,
 * that split along K into pieces of 1024 elements or more, as far as the
 * workspace holds their sums.
 * ---------------------------------------------------------------------- */
template <class E>
int too_large() {
  return fail(ZS_ERR_UNSUPPORTED, E::kOn ? "zs_mx_linear: too large for one launch%s"
                                         : "zs_mx_matmul: too large for one launch%s");
}

template <int AF, int CDT, int BM, int BN, int NW, class E>
int launch_tile(const MatmulArgs &a, uint32_t splits, const E &e, hipStream_t s) {
  const uint64_t tiles = (uint64_t)((a.m + BM - 1) / BM) * ((a.n + BN - 1) / BN);
  if (!fits(tiles, 64 * NW)) return too_large<E>();
  hipLaunchKernelGGL((matmul_tile_kernel<AF, CDT, BM, BN, NW, E>), dim3((unsigned)tiles, splits),
                     dim3(64 * NW), 0, s, a, e);
  return launch_result();
}

constexpr uint64_t kMaxMatmulK = 1ull << 22; /* byte offsets in a tile of 256 rows are 32 bits */
constexpr uint64_t kFullChip = 256; /* blocks that give every CU one */

/* Whether the thin kernel runs: every block reads all of A, which 32 rows of
 * B to a block repay for a few rows of A, or where tiles would leave half of
 * the CUs idle, or spend most of the two passes over an 8-bit A on rows that
 * are not there (32 x 32000 x 4096: 8-bit A 29 us, in tiles 31; 17 rows 23 and
 * 31; 4-bit A 20 us, in tiles 16). */
inline bool matmul_thin(uint64_t m, uint64_t n, bool wide_a) {
  return m <= 16 || (m <= 32 && (wide_a || n <= 128 * 128));
}

struct MatmulSplit {
  uint32_t splits, groups;   /* groups of 128 elements of K per split */
};

inline MatmulSplit matmul_split(uint64_t m, uint64_t n, uint64_t padded, uint64_t workspace_bytes) {
  const uint64_t tiles = (m + 127) / 128 * ((n + 127) / 128), groups = padded / ZS_MX_GROUP;
  uint64_t splits = kFullChip / tiles;
  if (splits > groups / 8) splits = groups / 8;
  if (splits > workspace_bytes / (m * n * 4)) splits = workspace_bytes / (m * n * 4);
  /* four at least: two pieces cost more than they save (512 x 4096 x 4096
   * 4-bit: 25 us against 16 in one), more pay (768 x 768 x 8192 8-bit A: 24
   * against 53; 65 x 4096 x 4096: 16 against 29) */
  if (matmul_thin(m, n, false) || splits < 4) return {1, (uint32_t)groups};
  const uint64_t each = (groups + splits - 1) / splits, four = (each + 3) / 4 * 4;
  return {(uint32_t)((groups + four - 1) / four), (uint32_t)four};
}

/* What a split product's first launch has for an epilogue: none, by a name of
 * its own in each of the sources that launch one. */
template <class E>
struct SplitEpilogue : NoEpilogue {};

template <int AF, int CDT, class E>
int launch_matmul(MatmulArgs a, const E &e, float *workspace, uint64_t workspace_bytes,
                  hipStream_t s) {
  constexpr uint64_t esz = CDT == ZS_FP32 ? 4 : 2;
  a.split_groups = a.padded / ZS_MX_GROUP;
  if (matmul_thin(a.m, a.n, AF == ZS_MX_E4M3)) {
    /* four results of a lane in one store */
    const int vec = aligned(a.c, 4 * esz) && a.ldc % 4 == 0;
    const uint32_t blocks = (a.n + 31) / 32;
    if (!fits(blocks, 64 * kThinWaves)) return too_large<E>();
    /* both halves of an 8-bit A in one instruction: 1 x 32000 x 4096 15.6 us,
     * in two 18.9; 4 rows 18.0 and 19.3; 16 rows 26.6 and 22.5 */
    if (AF == ZS_MX_E4M3 && a.m <= 4)
      hipLaunchKernelGGL((matmul_thin_kernel<AF, CDT, AF == ZS_MX_E4M3, E>), dim3(blocks),
                         dim3(64 * kThinWaves), 0, s, a, vec, e);
    else
      hipLaunchKernelGGL((matmul_thin_kernel<AF, CDT, false, E>), dim3(blocks), dim3(64 * kThinWaves),
                         0, s, a, vec, e);
    return launch_result();
  }
  constexpr int BM = AF == ZS_MX_E2M1 ? 256 : 128, BN = 256;
  if ((uint64_t)((a.m + BM - 1) / BM) * ((a.n + BN - 1) / BN) >= kFullChip)
    return launch_tile<AF, CDT, BM, BN, AF == ZS_MX_E2M1 ? 8 : 4>(a, 1, e, s);

  const MatmulSplit sp = matmul_split(a.m, a.n, a.padded, workspace_bytes);
  if (sp.splits < 2) return launch_tile<AF, CDT, 128, 128, 4>(a, 1, e, s);

  a.part = workspace;
  a.split_groups = sp.groups;
  if (int rc = launch_tile<AF, ZS_FP32, 128, 128, 4>(a, sp.splits, SplitEpilogue<E>{}, s)) return rc;
  const uint64_t all = (uint64_t)a.m * a.n;
  hipLaunchKernelGGL((matmul_join_kernel<CDT, E>), dim3((unsigned)((all + kBlock - 1) / kBlock)),
                     dim3(kBlock), 0, s, a, sp.splits, e);
  return launch_result();
}

}  // namespace zs_ops
#endif  // ZS_MATMUL_LAUNCH_H
