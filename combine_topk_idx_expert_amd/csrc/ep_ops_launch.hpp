// ep_ops_launch.hpp -- argument checks and launch configuration of the routing
// and int8 operators.
//
// Part of ep_api.hip's translation unit: it is included there, inside the
// anonymous namespace, after the error helpers (fail, EP_LAUNCHED) it uses.
#pragma once

constexpr int kCUs = 256;  // MI355X

// Calls f with the element-access type of an EP_TYPE_* value.
template <typename F>
ep_status with_type(int32_t type, F f) {
  switch (type) {
    case EP_TYPE_F32: return f(F32{});
    case EP_TYPE_BF16: return f(Bf16{});
    case EP_TYPE_F16: return f(F16{});
    default: return fail(EP_ERR_SHAPE, "unknown element type %d", type);
  }
}

uintptr_t type_bytes(int32_t type) { return type == EP_TYPE_F32 ? 4 : 2; }

ep_status validate_matmul(int64_t num_rows, int32_t num_groups, int32_t outer, uint32_t flags) {
  if (flags & ~(uint32_t)EP_MATMUL_GATED) return fail(EP_ERR_SHAPE, "unknown matmul flags 0x%x", flags);
  if (num_rows < 0 || num_groups < 0 || num_groups > EP_MAX_EXPERTS)
    return fail(EP_ERR_SHAPE, "bad sizes: %lld rows, %d groups (at most %d)", (long long)num_rows, num_groups,
                EP_MAX_EXPERTS);
  if (outer < 1 || outer > EP_MAX_MATMUL_OUTER || ((flags & EP_MATMUL_GATED) && outer % 2 != 0))
    return fail(EP_ERR_SHAPE, "outer %d must lie in [1, %d] and be even for a gated product", outer, EP_MAX_MATMUL_OUTER);
  if (num_rows >= (int64_t)1 << 31) return fail(EP_ERR_OVERFLOW, "num_rows %lld reaches 2^31", (long long)num_rows);
  return EP_OK;
}

ep_status validate_route(const ep_route_config* c, int32_t type, int64_t num_tokens, int64_t row_stride) {
  if (!c) return fail(EP_ERR_NULL, "route config is NULL");
  if (c->num_experts < 1 || c->num_experts > EP_MAX_EXPERTS)
    return fail(EP_ERR_SHAPE, "num_experts %d outside [1, %d]", c->num_experts, EP_MAX_EXPERTS);
  if (c->num_topk < 1 || c->num_topk > EP_MAX_TOPK)
    return fail(EP_ERR_SHAPE, "num_topk %d outside [1, %d]", c->num_topk, EP_MAX_TOPK);
  if (c->num_groups < 1 || c->num_groups > EP_MAX_ROUTE_GROUPS || c->num_experts % c->num_groups != 0)
    return fail(EP_ERR_SHAPE, "num_groups %d must divide num_experts %d and lie in [1, %d]", c->num_groups,
                c->num_experts, EP_MAX_ROUTE_GROUPS);
  if (c->topk_groups < 1 || c->topk_groups > c->num_groups)
    return fail(EP_ERR_SHAPE, "topk_groups %d outside [1, %d]", c->topk_groups, c->num_groups);
  if (c->num_topk > c->topk_groups * (c->num_experts / c->num_groups))
    return fail(EP_ERR_SHAPE, "num_topk %d exceeds the %d experts of topk_groups groups", c->num_topk,
                c->topk_groups * (c->num_experts / c->num_groups));
  if (c->score != EP_SCORE_SOFTMAX && c->score != EP_SCORE_SIGMOID)
    return fail(EP_ERR_SHAPE, "unknown score %d", c->score);
  if (c->group_score != EP_GROUP_MAX && c->group_score != EP_GROUP_TOP2)
    return fail(EP_ERR_SHAPE, "unknown group score %d", c->group_score);
  if (!(c->scale - c->scale == 0.0f)) return fail(EP_ERR_SHAPE, "scale must be finite");
  if (type != EP_TYPE_F32 && type != EP_TYPE_BF16 && type != EP_TYPE_F16)
    return fail(EP_ERR_SHAPE, "unknown element type %d", type);
  if (num_tokens < 0) return fail(EP_ERR_SHAPE, "num_tokens %lld < 0", (long long)num_tokens);
  if (num_tokens > 0 && row_stride < c->num_experts)
    return fail(EP_ERR_SHAPE, "row_stride %lld below num_experts %d", (long long)row_stride, c->num_experts);
  if (num_tokens > EP_MAX_ROUTE_TOKENS)
    return fail(EP_ERR_OVERFLOW, "num_tokens %lld above %d", (long long)num_tokens, EP_MAX_ROUTE_TOKENS);
  if (row_stride > ((int64_t)1 << 40)) return fail(EP_ERR_OVERFLOW, "row_stride %lld too large", (long long)row_stride);
  return EP_OK;
}

template <typename IO, int LPR, int VPL, int R>
ep_status launch_route_lanes(const RouteArgs& a, RouteLanes p, hipStream_t s) {
  constexpr int kRows = kWave / LPR;
  p.pad = p.seg != VPL || p.gs * a.G != p.seg * LPR;
  const size_t lds = std::max(((size_t)kRows * p.row_pitch + VPL) * sizeof(float), (size_t)a.E * sizeof(double));
  route_lanes_kernel<IO, LPR, VPL, R><<<(a.T + kRows - 1) / kRows, kWave, lds, s>>>(a, p);
  EP_LAUNCHED("route_lanes_kernel");
  return EP_OK;
}

template <typename IO, int LPR, int VPL>
ep_status launch_route_lanes(const RouteArgs& a, const RouteLanes& p, hipStream_t s) {
  return a.K <= 8 ? launch_route_lanes<IO, LPR, VPL, 1>(a, p, s) : launch_route_lanes<IO, LPR, VPL, 2>(a, p, s);
}

// Up to 512 experts and 16 choices: several rows a wave.  A group is 1, 2, 4 or 8
// lanes of eight, or of sixteen where eight lanes of 32 experts do not hold it;
// routers for which that does not come out, and wider ones, take one row a wave.
template <typename IO>
ep_status launch_route(const RouteArgs& a, hipStream_t s) {
  for (int lanes = 8; a.K <= 16 && lanes <= 16; lanes *= 2) {
    if (a.G > lanes) continue;
    RouteLanes p{};
    p.gs = a.E / a.G;
    while (a.G << (p.shift + 1) <= lanes && (a.G == 1 || p.shift < 3)) ++p.shift;
    const int wide = 1 << p.shift;
    p.seg = (p.gs + wide - 1) / wide;
    if (a.G == 1) p.seg = (p.seg + 3) / 4 * 4;
    if (p.seg > 32) continue;
    if (a.G == 1 || (p.gs == wide * p.seg && p.seg % 4 == 0)) {
      p.pitch = 4 * ((p.seg + 3) / 4 | 1);
      p.row_pitch = lanes * p.pitch;
      p.magic = (1 << 20) / p.seg + 1;
    } else {
      p.row_pitch = (a.E + 3) / 4 * 4;
    }
    p.bias_vec = p.seg % 4 == 0 && p.gs % 4 == 0 && !misaligned(a.bias, 16);
    if (lanes == 16) return launch_route_lanes<IO, 16, 32>(a, p, s);
    if (p.seg <= 8 && a.K <= 8) return launch_route_lanes<IO, 8, 8, 1>(a, p, s);
    if (p.seg <= 16) return launch_route_lanes<IO, 8, 16>(a, p, s);
    return launch_route_lanes<IO, 8, 32>(a, p, s);
  }
  const int waves = a.E > 2048 ? kRouteWaves / 2 : kRouteWaves;  // at most 64 KiB of LDS
  const int blocks = (a.T + waves - 1) / waves;
  route_kernel<IO><<<blocks, waves * kWave, (size_t)waves * a.E * sizeof(double), s>>>(a);
  EP_LAUNCHED("route_kernel");
  return EP_OK;
}

template <typename IO, int LPR>
ep_status launch_route_backward_lanes(const RouteBwdArgs& a, hipStream_t s) {
  constexpr int kRows = kWave / LPR, V = 16 / sizeof(typename IO::type);
  const bool dense = !a.sigmoid && !a.renorm;
  const int vec = a.E % V == 0;
  const size_t lds = (size_t)kRows * a.E * sizeof(float);
  const int blocks = (int)std::min<int64_t>((a.T + kRows - 1) / kRows, 16 * kCUs);
  const int pieces = (a.E / V + LPR - 1) / LPR;  // of a row, a lane
  if (dense && pieces <= 2)
    route_backward_lanes_kernel<IO, LPR, 2><<<blocks, kWave, lds, s>>>(a, vec);
  else if (dense && pieces <= 4)
    route_backward_lanes_kernel<IO, LPR, 4><<<blocks, kWave, lds, s>>>(a, vec);
  else if (dense && pieces <= 8)
    route_backward_lanes_kernel<IO, LPR, 8><<<blocks, kWave, lds, s>>>(a, vec);
  else
    route_backward_lanes_kernel<IO, LPR, 0><<<blocks, kWave, lds, s>>>(a, vec);
  EP_LAUNCHED("route_backward_lanes_kernel");
  return EP_OK;
}

// Up to 16 choices of 1024 experts: several rows a wave (at most 32 KiB of LDS).
template <typename IO>
ep_status launch_route_backward(const RouteBwdArgs& a, hipStream_t s) {
  if (a.E <= 1024 && a.K <= 8) return launch_route_backward_lanes<IO, 8>(a, s);
  if (a.E <= 1024 && a.K <= 16) return launch_route_backward_lanes<IO, 16>(a, s);
  const int blocks = (a.T + kRouteWaves - 1) / kRouteWaves;
  const size_t lds = (size_t)kRouteWaves * a.E * sizeof(float);
  route_backward_kernel<IO><<<blocks, kRouteWaves * kWave, lds, s>>>(a);
  EP_LAUNCHED("route_backward_kernel");
  return EP_OK;
}

template <typename IO, int WAVES>
ep_status launch_quantize_rows(const QuantArgs& a, int nc, hipStream_t s) {
  const int blocks = (int)((a.N * WAVES + 3) / 4);
  if (nc <= 1)
    quantize_rows_kernel<IO, WAVES, 1><<<blocks, 256, 0, s>>>(a);
  else if (nc <= 2)
    quantize_rows_kernel<IO, WAVES, 2><<<blocks, 256, 0, s>>>(a);
  else if (nc <= 4)
    quantize_rows_kernel<IO, WAVES, 4><<<blocks, 256, 0, s>>>(a);
  else
    quantize_rows_kernel<IO, WAVES, 8><<<blocks, 256, 0, s>>>(a);
  EP_LAUNCHED("quantize_rows_kernel");
  return EP_OK;
}

template <typename IO>
ep_status launch_quantize(const QuantArgs& a, hipStream_t s) {
  constexpr int V = 16 / sizeof(typename IO::type);
  const int chunks = a.H / V;
  const bool whole = a.H % V == 0;
  if (whole && a.N >= 4 * kCUs && chunks <= 8 * kWave) return launch_quantize_rows<IO, 1>(a, (chunks + 63) / 64, s);
  if (whole && chunks <= 8 * 4 * kWave) return launch_quantize_rows<IO, 4>(a, (chunks + 255) / 256, s);
  quantize_kernel<IO><<<(int)a.N, kQuantThreads, 0, s>>>(a);
  EP_LAUNCHED("quantize_kernel");
  return EP_OK;
}

template <typename IO, bool GATED, int BM, int BN, int WM, int WN, bool HALVES>
ep_status launch_matmul_tile(const MatmulArgs& a, hipStream_t s) {
  typedef TileShape<BM, BN, WM, WN> S;
  const int bc = GATED ? BN / 2 : BN;
  const int64_t n_tiles = (a.width + bc - 1) / bc;
  const int64_t most = (a.M / BM + a.G) * n_tiles;  // each group's last row tile may be partly filled
  if (most >= (int64_t)1 << 31) return fail(EP_ERR_OVERFLOW, "product of %lld tiles is too large", (long long)most);
  const int grid = (int)std::min<int64_t>(most, kCUs);
  matmul_tile_kernel<IO, GATED, BM, BN, WM, WN, HALVES><<<grid, S::kThreads, S::lds(a.G), s>>>(a, (int)n_tiles);
  EP_LAUNCHED("matmul_tile_kernel");
  return EP_OK;
}

template <typename IO, bool GATED, int MT, int NT, int KW, int S>
ep_status launch_matmul_split(const MatmulArgs& a, hipStream_t s) {
  const int bc = (GATED ? NT / 2 : NT) * 16;
  const int64_t nb = (a.width + bc - 1) / bc;
  // row tiles side by side; a workgroup takes several where there are more.  For
  // groups: twice the mean, or what fills the card
  int64_t y = std::min<int64_t>((std::min(a.M, a.most) + 16 * MT - 1) / (16 * MT), 4096);
  if (a.row_start)
    y = std::min(y, std::max<int64_t>((2 * a.M / a.G + 16 * MT - 1) / (16 * MT), 32 * kCUs / (nb * a.G) + 1));
  matmul_split_kernel<IO, GATED, MT, NT, KW, S><<<dim3((unsigned)nb, (unsigned)y, a.G), KW * kWave, 0, s>>>(a);
  EP_LAUNCHED("matmul_split_kernel");
  return EP_OK;
}

// Which kernel (both sides measured on MI355X):
//  - tiles of 256 x 256 once they fill three quarters of the CUs; below that
//    tiles of 128 x 256 while they fill three eighths (2048 x 7168 x 4096 gated: 67
//    against 82 us; 8192 x 8192 x 8192: 256 x 256 by 10%);
//  - below that, and for at most 64 rows whatever the width, the split over the inner
//    size (512 x 7168 x 4096 gated: 23 us against 54 and 79; 64 rows: 9 against 44 and
//    49; 1 x 7168 x 49152: 63 against 88 and 90, 64 rows of it 87 against 91 and 93).
// Groups: their sizes are on the device.  A group of at most kFewRows rows is
// the split's and a larger one the tiles'; each launch passes over the others'
// groups.  No second launch where large groups cannot fill more than half of the tiles'
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
template <typename IO, bool GATED, int MT, int NT>
ep_status launch_matmul_split(const MatmulArgs& a, int64_t blocks, hipStream_t s) {
  const bool stream = a.K >= 2048 && (int64_t)a.G * a.N * a.K >= (int64_t)8 << 20;
  return stream && (MT == 1 || blocks <= kCUs) ? launch_matmul_split<IO, GATED, MT, NT, 4, 2>(a, s)
                                               : launch_matmul_split<IO, GATED, MT, NT, 2, 2>(a, s);
}

template <typename IO, bool GATED>
ep_status launch_matmul_few(const MatmulArgs& a, hipStream_t s) {
  constexpr int kShapes[5][2] = {{1, 2}, {1, 4}, {2, 2}, {2, 4}, {4, 4}};
  const int64_t mean = std::min(a.M / a.G + (a.M % a.G != 0), a.most);
  int64_t least = INT64_MAX, blocks = 0;
  int best = 0;
  for (int i = 0; i < 5; ++i) {
    const int rows = 16 * kShapes[i][0], cols = (GATED ? 8 : 16) * kShapes[i][1];
    const int64_t n = (mean + rows - 1) / rows * a.G * ((a.width + cols - 1) / cols);
    const int64_t cost = (n + kCUs - 1) / kCUs * (kShapes[i][0] + kShapes[i][1]);
    if (cost > least) continue;  // (of equals the larger one)
    least = cost;
    blocks = n;
    best = i;
  }
  switch (best) {
    case 0: return launch_matmul_split<IO, GATED, 1, 2>(a, blocks, s);
    case 1: return launch_matmul_split<IO, GATED, 1, 4>(a, blocks, s);
    case 2: return launch_matmul_split<IO, GATED, 2, 2>(a, blocks, s);
    case 3: return launch_matmul_split<IO, GATED, 2, 4>(a, blocks, s);
    default: return launch_matmul_split<IO, GATED, 4, 4>(a, blocks, s);
  }
}

// EP_KERNEL_* of the launches for M rows in G groups (0: dense) and `width` columns of out.
uint32_t matmul_kernels(int64_t M, int G, int width, bool gated) {
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

template <typename IO, bool GATED>
ep_status launch_matmul(MatmulArgs a, hipStream_t s) {
  const uint32_t kernels = matmul_kernels(a.M, a.row_start ? a.G : 0, a.width, GATED);
  a.least = 0;
  a.most = a.M;
  if (kernels & EP_KERNEL_SPLIT) {
    MatmulArgs few = a;
    if (kernels != EP_KERNEL_SPLIT) few.most = kFewRows;
    const ep_status st = launch_matmul_few<IO, GATED>(few, s);
    if (st != EP_OK || kernels == EP_KERNEL_SPLIT) return st;
    a.least = kFewRows + 1;
  }
  if (kernels & EP_KERNEL_TILES_256) return launch_matmul_tile<IO, GATED, 256, 256, 2, 4, true>(a, s);
  return launch_matmul_tile<IO, GATED, 128, 256, 2, 4, false>(a, s);
}
