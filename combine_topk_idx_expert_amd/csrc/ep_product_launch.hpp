// ep_product_launch.hpp -- argument checks and launch configuration of the products.
#pragma once

#include <algorithm>

#include "ep_host.hpp"
#include "ep_int8_tile.hpp"
#include "ep_product.hpp"
#include "ep_product_tile.hpp"

namespace ep {

inline ep_status validate_matmul(int64_t num_rows, int32_t num_groups, int32_t outer, uint32_t flags,
                                 uint32_t known = EP_MATMUL_GATED) {
  if (flags & ~known) return fail(EP_ERR_SHAPE, "unknown matmul flags 0x%x", flags);
  if (num_rows < 0 || num_groups < 0 || num_groups > EP_MAX_EXPERTS)
    return fail(EP_ERR_SHAPE, "bad sizes: %lld rows, %d groups (at most %d)", (long long)num_rows, num_groups,
                EP_MAX_EXPERTS);
  if (outer < 1 || outer > EP_MAX_MATMUL_OUTER || ((flags & EP_MATMUL_GATED) && outer % 2 != 0))
    return fail(EP_ERR_SHAPE, "outer %d must lie in [1, %d] and be even for a gated product", outer, EP_MAX_MATMUL_OUTER);
  if (num_rows >= (int64_t)1 << 31) return fail(EP_ERR_OVERFLOW, "num_rows %lld reaches 2^31", (long long)num_rows);
  return EP_OK;
}

template <typename AR, typename IO, bool GATED, int BM, bool HALVES>
ep_status launch_matmul_tile(const MatmulArgs& a, hipStream_t s) {
  const int bc = GATED ? 128 : 256;
  const int64_t n_tiles = (a.width + bc - 1) / bc;
  const int64_t most = (a.M / BM + a.G) * n_tiles;  // each group's last row tile may be partly filled
  if (most >= (int64_t)1 << 31) return fail(EP_ERR_OVERFLOW, "product of %lld tiles is too large", (long long)most);
  const int grid = (int)std::min<int64_t>(most, kCUs);
  if constexpr (AR::kScales == kRowScales) {
    typedef TileShape<BM, 256, 2, 4> S;
    matmul_tile_kernel<IO, GATED, BM, 256, 2, 4, HALVES><<<grid, S::kThreads, S::lds(a.G), s>>>(a, (int)n_tiles);
    EP_LAUNCHED("matmul_tile_kernel");
  } else {
    typedef StepShape<BM, 256, 2, 4, AR::kScales == kBlockScales> S;
    product_tile_kernel<AR, IO, GATED, BM, 256, 2, 4, HALVES><<<grid, S::kThreads, S::lds(a.G), s>>>(a, (int)n_tiles);
    EP_LAUNCHED("product_tile_kernel");
  }
  return EP_OK;
}

template <typename AR, typename IO, bool GATED, int MT, int NT, int KW, int S>
ep_status launch_matmul_split(const MatmulArgs& a, hipStream_t s) {
  const int bc = (GATED ? NT / 2 : NT) * 16;
  const int64_t nb = (a.width + bc - 1) / bc;
  // row tiles side by side; a workgroup takes several where there are more.  For
  // groups: twice the mean, or what fills the card
  int64_t y = std::min<int64_t>((std::min(a.M, a.most) + 16 * MT - 1) / (16 * MT), 4096);
  if (a.row_start)
    y = std::min(y, std::max<int64_t>((2 * a.M / a.G + 16 * MT - 1) / (16 * MT), 32 * kCUs / (nb * a.G) + 1));
  matmul_split_kernel<AR, IO, GATED, MT, NT, KW, S><<<dim3((unsigned)nb, (unsigned)y, a.G), KW * kWave, 0, s>>>(a);
  EP_LAUNCHED("matmul_split_kernel");
  return EP_OK;
}

// Which kernel (both sides measured on MI355X with int8; E4M3 and 16-bit products take the same
// rules unmeasured, but for tall_tiles below):
//  - tiles of 256 x 256 once they fill three quarters of the CUs; below that
//    tiles of 128 x 256 while they fill three eighths (2048 x 7168 x 4096 gated: 67
//    against 82 us; 8192 x 8192 x 8192: 256 x 256 by 10%);
//  - below that, and for at most 64 rows whatever the width, the split over the inner
//    size (512 x 7168 x 4096 gated: 23 us against 54 and 79; 64 rows: 9 against 44 and
//    49; 1 x 7168 x 49152: 63 against 88 and 90, 64 rows of it 87 against 91 and 93).
// Groups: their sizes are on the device.  A group of at most kFewRows rows is
// the split's and a larger one the tiles'; each launch passes over the others'
// groups.  (The mean counts the groups' padding.)  No second launch where large groups cannot fill more than half of the tiles'
// grid (8 groups of 72 rows, 7168 x 4096 gated: 72 us by the split alone, 84 by both),
// or three eighths for tall groups, whose rows the split takes 64 at a time (8 of 1696,
// 4672 x 318 gated: 46 us by tiles, 80 by the split); nor a first one where the mean
// is so large that few groups are small.  129 random shapes (2 to 64 groups, inner 320
// to 7168): with 96 to 128 tiles of large groups, tiles take 1.28 times the split's time
// for means of up to 128 rows, 1.03 for 129 to 199, 0.72 above; with fewer 1.22, 1.22 and
// 0.97, with up to 192 1.00, 0.85 and 0.72.  The rule is within 10% of the fastest of the
// three in 106 of them and 4% off on average (at worst 1.6 times: 32 groups of 112
// rows, 2048 x 256, by the split 35 us, by tiles 22).
constexpr int64_t kFewRows = 64;

// The split's tile, MT x NT sixteens of rows and channels.  Its time is that of the
// loads, MT + NT for each step of a workgroup, on the CU with the most workgroups:
// the shape for which that is least.  1 x 7168 x 4096 gated: 1 x 2 7.4 us, 1 x 4 9.0;
// 64 rows: 2 x 2 9.0, 1 x 2 10.5, 2 x 4 9.8, 4 x 4 12.6; 512 rows: 4 x 4 23, 2 x 4 35;
// 3475 x 6432 x 99: 2 x 4 14, 4 x 4 18.
// Two waves a workgroup leave room for several workgroups a CU.  Four are better
// where weights that no cache holds stream through a long inner size (one row: 7.4
// against 9.4 us; 32 groups of 3 rows: 154 against 160; from the L2, 8 groups of 79
// rows, 3904 x 78: 9.3 against 7.1) and a CU has one workgroup or small ones (512
// rows, two a CU: 27 against 23).
struct SplitShape {
  int rows, cols, waves;  // sixteens of rows and channels
};

inline SplitShape split_shape(const MatmulArgs& a, bool gated) {
  constexpr int kShapes[5][2] = {{1, 2}, {1, 4}, {2, 2}, {2, 4}, {4, 4}};
  const int64_t mean = std::min(a.M / a.G + (a.M % a.G != 0), a.most);
  int64_t least = INT64_MAX, blocks = 0;
  SplitShape best{};
  for (const auto& shape : kShapes) {
    const int rows = 16 * shape[0], cols = (gated ? 8 : 16) * shape[1];
    const int64_t n = (mean + rows - 1) / rows * a.G * ((a.width + cols - 1) / cols);
    const int64_t cost = (n + kCUs - 1) / kCUs * (shape[0] + shape[1]);
    if (cost > least) continue;  // (of equals the larger one)
    least = cost;
    blocks = n;
    best = SplitShape{shape[0], shape[1], 2};
  }
  const bool stream = a.K >= 2048 && (int64_t)a.G * a.N * a.K >= (int64_t)8 << 20;
  if (stream && (best.rows == 1 || blocks <= kCUs)) best.waves = 4;
  return best;
}

template <typename AR, typename IO, bool GATED, int MT, int NT>
ep_status launch_matmul_split(const MatmulArgs& a, int waves, hipStream_t s) {
  return waves == 4 ? launch_matmul_split<AR, IO, GATED, MT, NT, 4, 2>(a, s)
                    : launch_matmul_split<AR, IO, GATED, MT, NT, 2, 2>(a, s);
}

template <typename AR, typename IO, bool GATED>
ep_status launch_matmul_few(const MatmulArgs& a, hipStream_t s) {
  const SplitShape t = split_shape(a, GATED);
  if (t.rows == 1)
    return t.cols == 2 ? launch_matmul_split<AR, IO, GATED, 1, 2>(a, t.waves, s)
                       : launch_matmul_split<AR, IO, GATED, 1, 4>(a, t.waves, s);
  if (t.rows == 2)
    return t.cols == 2 ? launch_matmul_split<AR, IO, GATED, 2, 2>(a, t.waves, s)
                       : launch_matmul_split<AR, IO, GATED, 2, 4>(a, t.waves, s);
  return launch_matmul_split<AR, IO, GATED, 4, 4>(a, t.waves, s);
}

// EP_KERNEL_* of the launches for M rows in G groups (0: dense) and `width` columns of out.
inline uint32_t matmul_kernels(int64_t M, int G, int width, bool gated) {
  const int bc = gated ? 128 : 256;
  const int64_t n_tiles = (width + bc - 1) / bc;
  if (G == 0) {
    if (M <= kFewRows) return EP_KERNEL_SPLIT;
    if ((M + 255) / 256 * n_tiles >= 3 * kCUs / 4) return EP_KERNEL_TILES_256;
    if ((M + 127) / 128 * n_tiles >= 3 * kCUs / 8) return EP_KERNEL_TILES_128;
    return EP_KERNEL_SPLIT;
  }
  const int64_t mean = M / G;
  // row tiles that large groups can fill: a tile has more than kFewRows rows
  const int64_t large = std::min(M / 256 + G, M / (kFewRows + 1));
  if (mean <= 2 * kFewRows ? large * n_tiles <= kCUs / 2 : large * n_tiles < 3 * kCUs / 8) return EP_KERNEL_SPLIT;
  return ((M / 256 + G) * n_tiles >= 3 * kCUs / 4 ? EP_KERNEL_TILES_256 : EP_KERNEL_TILES_128) |
         (mean < 4 * kFewRows ? EP_KERNEL_SPLIT : 0);
}

// E4M3 and 16-bit dense products in tiles: the height whose rounds over the CUs cost less.  A
// step of 256 rows takes 1.7 (E4M3 1.9) times one of 128 (22240 x 2112 x 326 gated, 174 or 348
// tiles: 52 us by 256 rows, 59 by 128; 1003 x 2048 x 7168, 112 or 224: 36 by 128).
inline bool tall_tiles(int64_t M, int64_t n_tiles) {
  const int64_t tall = ((M + 255) / 256 * n_tiles + kCUs - 1) / kCUs, flat = ((M + 127) / 128 * n_tiles + kCUs - 1) / kCUs;
  return 17 * tall <= 10 * flat;
}

// EP_KERNEL_* of a product's launches: matmul_kernels, and for E4M3 and 16-bit rows the
// height above.  (bf16 fragments of E4M3 codes have no registers left for 256 rows.)
template <typename AR>
uint32_t product_kernels(int64_t M, int G, int width, bool gated) {
  uint32_t kernels = matmul_kernels(M, G, width, gated);
  if (AR::kScales != kRowScales && G == 0 && kernels != EP_KERNEL_SPLIT)
    kernels = tall_tiles(M, (width + (gated ? 127 : 255)) / (gated ? 128 : 256)) ? EP_KERNEL_TILES_256
                                                                               : EP_KERNEL_TILES_128;
  if (std::is_same_v<AR, Fp8ExactMath> && (kernels & EP_KERNEL_TILES_256))
    kernels ^= EP_KERNEL_TILES_256 | EP_KERNEL_TILES_128;
  return kernels;
}

template <typename AR, typename IO, bool GATED>
ep_status launch_matmul(MatmulArgs a, hipStream_t s) {
  const uint32_t kernels = product_kernels<AR>(a.M, a.row_start ? a.G : 0, a.width, GATED);
  a.least = 0;
  a.most = a.M;
  if (kernels & EP_KERNEL_SPLIT) {
    MatmulArgs few = a;
    if (kernels != EP_KERNEL_SPLIT) few.most = kFewRows;
    const ep_status st = launch_matmul_few<AR, IO, GATED>(few, s);
    if (st != EP_OK || kernels == EP_KERNEL_SPLIT) return st;
    a.least = kFewRows + 1;
  }
  if constexpr (!std::is_same_v<AR, Fp8ExactMath>)
    if (kernels & EP_KERNEL_TILES_256) return launch_matmul_tile<AR, IO, GATED, 256, true>(a, s);
  return launch_matmul_tile<AR, IO, GATED, 128, false>(a, s);
}

}  // namespace ep
