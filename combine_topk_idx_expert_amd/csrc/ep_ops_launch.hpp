// ep_ops_launch.hpp -- argument checks and launch configuration of the routing
// and int8 operators.
//
// Part of ep_api.hip's translation unit: it is included there, inside the
// anonymous namespace, after the error helpers (fail, EP_LAUNCHED) it uses.
#pragma once

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
  if (num_tokens * c->num_topk >= ((int64_t)1 << 31) || num_tokens >= ((int64_t)1 << 31))
    return fail(EP_ERR_OVERFLOW, "num_tokens * num_topk reaches 2^31");
  if (row_stride > ((int64_t)1 << 40)) return fail(EP_ERR_OVERFLOW, "row_stride %lld too large", (long long)row_stride);
  return EP_OK;
}

template <typename IO>
ep_status launch_route(const RouteArgs& a, hipStream_t s) {
  const int waves = a.E > 2048 ? kRouteWaves / 2 : kRouteWaves;  // at most 64 KiB of LDS
  const int blocks = (a.T + waves - 1) / waves;
  route_kernel<IO><<<blocks, waves * kWave, (size_t)waves * a.E * sizeof(double), s>>>(a);
  EP_LAUNCHED("route_kernel");
  return EP_OK;
}

template <typename IO>
ep_status launch_route_backward(const RouteBwdArgs& a, hipStream_t s) {
  const int blocks = (a.T + kRouteWaves - 1) / kRouteWaves;
  const size_t lds = (size_t)kRouteWaves * a.E * sizeof(float);
  route_backward_kernel<IO><<<blocks, kRouteWaves * kWave, lds, s>>>(a);
  EP_LAUNCHED("route_backward_kernel");
  return EP_OK;
}

template <typename IO>
ep_status launch_quantize(const QuantArgs& a, hipStream_t s) {
  quantize_kernel<IO><<<(int)a.N, kQuantThreads, 0, s>>>(a);
  EP_LAUNCHED("quantize_kernel");
  return EP_OK;
}

template <typename IO, bool GATED, int BM, int BN, int WM, int WN>
ep_status launch_matmul_tile(const MatmulArgs& a, int per_cu, hipStream_t s) {
  typedef TileShape<BM, BN, WM, WN> S;
  const int bc = GATED ? BN / 2 : BN;
  const int64_t n_tiles = (a.width + bc - 1) / bc;
  const int64_t most = (a.M / BM + a.G) * n_tiles;  // each group's last row tile may be partly filled
  if (most >= (int64_t)1 << 31) return fail(EP_ERR_OVERFLOW, "product of %lld tiles is too large", (long long)most);
  const int grid = (int)std::min<int64_t>(most, 256 * per_cu);
  matmul_tile_kernel<IO, GATED, BM, BN, WM, WN><<<grid, S::kThreads, S::lds(a.G), s>>>(a, (int)n_tiles);
  EP_LAUNCHED("matmul_tile_kernel");
  return EP_OK;
}

template <typename IO, bool GATED>
ep_status launch_matmul(const MatmulArgs& a, hipStream_t s) {
  if (a.M >= (int64_t)96 * a.G) return launch_matmul_tile<IO, GATED, 256, 256, 2, 4>(a, 1, s);
  const int64_t nb = (a.width + 63) / 64;
  const int64_t tiles = (a.M + kRowTile - 1) / kRowTile;
  const int z = (int)std::min<int64_t>(a.row_start ? (tiles + a.G - 1) / a.G : tiles, 4096);
  matmul_rows_kernel<IO, GATED><<<dim3((unsigned)nb, a.G, z), 256, 0, s>>>(a);
  EP_LAUNCHED("matmul_rows_kernel");
  return EP_OK;
}
